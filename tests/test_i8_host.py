"""CPU checks of the 8-bit integer operators and the router by groups: refusals
of the C ABI and of the binding before any device work, and the plain forms the
GPU tests use against brute force and differences."""
from __future__ import annotations

import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _i8
from tests import test_gpu_i8 as shapes

P = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced
P8 = ctypes.c_void_p((1 << 20) + 8)
P2 = ctypes.c_void_p((1 << 20) + 2)
P1 = ctypes.c_void_p((1 << 20) + 1)
N0 = ctypes.c_void_p(0)

EINVAL, EUNSUP = dbs.DBS_EINVAL, dbs.DBS_EUNSUPPORTED


def _refused(name, args, want):
    L = dbs.lib()
    assert getattr(L, name)(*args, N0) == want
    assert L.dbs_last_error().decode() != ""


# type, x, M, K, codes, scales
@pytest.mark.parametrize("args", [
    (0, N0, 4, 8, P, P), (0, P, 4, 8, N0, P), (0, P, 4, 8, P, N0), (2, P, 4, 8, P, P), (0, P, 0, 8, P, P),
    (0, P, 4, 0, P, P), (0, P, (1 << 25) + 1, 8, P, P), (0, P, 4, (1 << 21) + 1, P, P), (0, P2, 4, 8, P, P),
    (1, P1, 4, 8, P, P), (1, P, 4, 8, P, P2),
])
def test_quant_refusals(args):
    _refused("quant_i8", args, EINVAL)


# type, A, sA, B, sB, D, M, N, K
@pytest.mark.parametrize("args", [
    (0, N0, P, P, P, P, 4, 8, 16), (0, P, N0, P, P, P, 4, 8, 16), (0, P, P, N0, P, P, 4, 8, 16),
    (0, P, P, P, N0, P, 4, 8, 16), (0, P, P, P, P, N0, 4, 8, 16), (2, P, P, P, P, P, 4, 8, 16),
    (0, P, P, P, P, P, 0, 8, 16), (0, P, P, P, P, P, 4, 0, 16), (0, P, P, P, P, P, 4, 8, 0),
    (0, P, P, P, P, P, 4, 8, 24), (0, P, P, P, P, P, 4, 8, 1 << 17), (0, P, P, P, P, P, (1 << 25) + 1, 8, 16),
    (0, P, P, P, P, P, 4, (1 << 21) + 1, 16), (0, P8, P, P, P, P, 4, 8, 16), (0, P, P2, P, P, P, 4, 8, 16),
    (0, P, P, P8, P, P, 4, 8, 16), (0, P, P, P, P2, P, 4, 8, 16), (0, P, P, P, P, P2, 4, 8, 16),
    (1, P, P, P, P, P1, 4, 8, 16),
])
def test_product_refusals(args):
    _refused("gemm_i8", args, EINVAL)


# X, sX, W, sW, D, offsets, rows, T, M, E, N, K
@pytest.mark.parametrize("args,want", [
    ((N0, P, P, P, P, P, P, 4, 8, 2, 16, 16), EINVAL), ((P, N0, P, P, P, P, P, 4, 8, 2, 16, 16), EINVAL),
    ((P, P, P, P, P, N0, P, 4, 8, 2, 16, 16), EINVAL), ((P, P, P, P, P, P, P, 0, 8, 2, 16, 16), EINVAL),
    ((P, P, P, P, P, P, P, 4, 0, 2, 16, 16), EINVAL), ((P, P, P, P, P, P, P, 4, 8, 0, 16, 16), EINVAL),
    ((P, P, P, P, P, P, P, 4, 8, 1025, 16, 16), EINVAL), ((P, P, P, P, P, P, P, 4, 8, 2, 16, 8), EINVAL),
    ((P, P, P, P, P, P, N0, 4, 8, 2, 16, 16), EINVAL),                  # sorted, T != M
    ((P8, P, P, P, P, P, P, 4, 8, 2, 16, 16), EINVAL), ((P, P2, P, P, P, P, P, 4, 8, 2, 16, 16), EINVAL),
    ((P, P, P8, P, P, P, P, 4, 8, 2, 16, 16), EINVAL), ((P, P, P, P2, P, P, P, 4, 8, 2, 16, 16), EINVAL),
    ((P, P, P, P, P1, P, P, 4, 8, 2, 16, 16), EINVAL), ((P, P, P, P, P, P2, P, 4, 8, 2, 16, 16), EINVAL),
    ((P, P, P, P, P, P, P2, 4, 8, 2, 16, 16), EINVAL), ((P, P, P, P, P, P, P, 4, 8, 2, 16, 1 << 17), EINVAL),
    ((P, P, P, P, P, P, P, 1 << 25, 8, 2, 16, 128), EUNSUP),            # a 4 GiB gathered X
])
def test_experts_product_refusals(args, want):
    _refused("gemm_moe_i8", args, want)
    _refused("gemm_moe_swiglu_i8", args, want)


def test_limits_of_size():
    _refused("gemm_moe_swiglu_i8", (P, P, P, P, P, P, P, 4, 8, 2, (1 << 20) + 1, 16), EINVAL)
    _refused("gemm_moe_swiglu_i8", (P, P, P, P, P, P, P, 4, 8, 2, 1 << 14, 1 << 16), EUNSUP)      # 2 GiB of matrices
    _refused("gemm_i8", (1, P, P, P, P, P, 1 << 25, 1 << 16, 16), EUNSUP)                         # 2^19 x 2^11 tiles
    assert "tiles" in dbs.lib().dbs_last_error().decode()


def _route(type=0, logits=P, bias=N0, T=4, E=8, k=2, score=1, groups=2, kept=1, best=2, renorm=1, scale=1.0, experts=P,
           weights=P, offsets=P, rows=P, slots=P, ws=N0, n=0):
    return (type, logits, bias, T, E, k, score, groups, kept, best, renorm, scale, experts, weights, offsets, rows,
            slots, ws, n)


@pytest.mark.parametrize("more,want", [
    (dict(logits=N0), EINVAL), (dict(type=2), EINVAL), (dict(T=0), EINVAL), (dict(E=0), EINVAL), (dict(k=0), EINVAL),
    (dict(k=9), EINVAL), (dict(E=1026), EINVAL), (dict(E=64, k=17), EUNSUP), (dict(T=1 << 60, k=2), EINVAL),
    (dict(score=2), EINVAL), (dict(groups=0), EINVAL), (dict(groups=3), EINVAL), (dict(groups=16), EINVAL),
    (dict(kept=0), EINVAL), (dict(kept=3), EINVAL), (dict(best=0), EINVAL), (dict(best=3), EINVAL),
    (dict(k=5), EINVAL),                                                # more than the kept groups have
    (dict(E=64, groups=32, kept=8), EUNSUP),                            # more than 16 groups
    (dict(E=1023, groups=11, kept=11), EUNSUP),                         # 93 experts to a lane
    (dict(renorm=2), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(experts=N0), EINVAL), (dict(weights=P2), EINVAL), (dict(slots=N0), EINVAL), (dict(bias=P2), EINVAL),
    (dict(logits=P2), EINVAL), (dict(T=65), EINVAL), (dict(T=65, ws=P, n=4), EINVAL), (dict(T=65, ws=P8, n=1 << 20), EINVAL),
])
def test_route_grouped_refusals(more, want):
    _refused("moe_route_grouped", _route(**more), want)


def test_route_grouped_workspace_sizes():
    ws = dbs.lib().moe_route_grouped_workspace
    assert ws(64, 128, 8) == 0 and ws(0, 8, 2) == 0 and ws(100, 8, 9) == 0 and ws(100, 2000, 2) == 0
    # rows of bytes for 16, 32 or 64 tokens, of 32-bit counts and their totals above 16384
    assert ws(65, 8, 2) == 5 * 16 and ws(4096, 160, 2) == 256 * 160 and ws(4097, 161, 2) == 129 * 176
    assert ws(16384, 256, 8) == 256 * 256 and ws(16385, 3, 2) == 258 * 3 * 4


# type, logits, T, E, k, score, renorm, scale, experts, dweights, dlogits
@pytest.mark.parametrize("args", [
    (0, N0, 4, 8, 2, 1, 1, 1.0, P, P, P), (0, P, 4, 8, 2, 2, 1, 1.0, P, P, P), (0, P, 4, 8, 2, 1, 2, 1.0, P, P, P),
    (0, P, 4, 8, 2, 1, 1, float("inf"), P, P, P), (0, P, 4, 8, 9, 1, 1, 1.0, P, P, P), (0, P, 4, 8, 2, 1, 1, 1.0, N0, P, P),
    (0, P, 4, 8, 2, 1, 1, 1.0, P, N0, P), (0, P, 4, 8, 2, 1, 1, 1.0, P, P, N0), (0, P, 4, 8, 2, 1, 1, 1.0, P, P, P2),
    (5, P, 4, 8, 2, 1, 1, 1.0, P, P, P),
])
def test_route_grouped_bwd_refusals(args):
    _refused("moe_route_grouped_bwd", args, EINVAL)


def test_binding_refuses_what_is_not_right():
    x, q = torch.zeros(4, 16), torch.zeros(4, 16, dtype=torch.int8)
    s, i = torch.zeros(4), torch.zeros(4, 2, dtype=torch.int32)
    w, sw, off = q[None].repeat(2, 1, 1), torch.zeros(2, 4), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: dbs.quant_i8(x), lambda: dbs.gemm_i8(q, s, q, s), lambda: dbs.gemm_moe_i8(q, s, w, sw, off),
                 lambda: dbs.gemm_moe_swiglu_i8(q, s, w, sw, off), lambda: dbs.moe_route_grouped(x, 2),
                 lambda: dbs.moe_route_grouped_backward(x, i, torch.zeros(4, 2))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: dbs.quant_i8(None), lambda: dbs.gemm_i8(None, s, q, s), lambda: dbs.moe_route_grouped(x, 2.5)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: dbs.quant_i8(x[0]), lambda: dbs.gemm_i8(q[0], s, q, s),
                 lambda: dbs.gemm_moe_i8(q, s, q, sw, off)):
        with pytest.raises(ValueError, match="dimensions"):
            call()
    with pytest.raises(ValueError, match="even"):
        dbs.gemm_moe_swiglu_i8(q, s, w[:, :3], sw[:, :3], off)


# ------------------------------------------------------------- the plain forms


def test_plain_quant_against_fractions():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 24)).astype(np.float32)
    x[1] = np.arange(24) * 0.5                            # many ties: 127 x / amax at halves
    x[1, 0] = 127.0
    x[2] = 0
    x[3] *= np.float32(1e-40)
    x[4] = np.float32(3e38) * np.sign(x[4])
    x[5] = np.where(np.arange(24) % 2, 1.0, 2.0)          # 63.5
    codes, scales = _i8.quant(x.astype(np.float64))
    for m in range(len(x)):
        amax = max(abs(Fraction(float(v))) for v in x[m])
        for k in range(x.shape[1]):
            want = 0 if amax == 0 else round(127 * Fraction(float(x[m, k])) / amax)      # (ties to even)
            assert codes[m, k] == want, (m, k)
    assert (codes[5][1::2] == 64).all() and scales[2] == 0


def _brute_choice(c, there, groups, kept, best, k):
    E = len(c)
    left = {e for e in range(E) if there[e]}
    if kept < groups:
        score = []
        for g in range(groups):
            mine = [e for e in left if e * groups // E == g]
            total, n = 0.0, 0
            while mine and n < best:
                top = max(mine, key=lambda e: c[e])
                total, n = total + c[top], n + 1
                mine.remove(top)
            score.append(total if n else None)
        keep = set()
        for _ in range(kept):
            able = [g for g in range(groups) if score[g] is not None and g not in keep]
            if able:
                keep.add(max(able, key=lambda g: (score[g], -g)))
        left = {e for e in left if e * groups // E in keep}
    out = []
    while left and len(out) < k:
        top = max(left, key=lambda e: (c[e], -e))
        out.append(top)
        left.remove(top)
    return out + [-1] * (k - len(out))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,kept,best", [(1, 1, 2), (4, 2, 2), (4, 1, 1), (3, 3, 2)])
def test_plain_choice_against_brute_force(kind, groups, kept, best):
    rng = np.random.default_rng(2)
    x = np.round(rng.standard_normal((30, 12)) * 4) / 4          # ties
    x[rng.random(x.shape) < 0.3] = -np.inf
    x[0] = -np.inf
    bias = np.round(rng.standard_normal(12) * 8) / 8
    bias[5] = -np.inf
    got = _i8.choose(x, 3, bias, groups, kept, best, kind)
    for t in range(len(x)):
        s = _i8.scores(x[t], kind)
        there = (x[t] > -np.inf) & (bias > -np.inf)
        c = np.where(there, s + np.where(bias > -np.inf, bias, 0), 0)
        assert got[t].tolist() == _brute_choice(c, there, groups, kept, best, 3)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_gradient_against_differences(kind, renorm):
    rng = np.random.default_rng(3)
    x, d = rng.standard_normal((4, 8)) * 2, rng.standard_normal((4, 3))
    experts = _i8.choose(x, 3, None, 1, 1, 2, kind)
    g = _i8.grouped_grad(x, experts, d, kind, renorm, 1.7)
    h = 1e-5
    for t in range(4):
        for e in range(8):
            y, z = x.copy(), x.copy()
            y[t, e] += h
            z[t, e] -= h
            (wy, _), (wz, _) = (_i8.weights(v, experts, kind, renorm, 1.7) for v in (y, z))
            assert abs(((wy - wz) * d).sum() / (2 * h) - g[t, e]) < 1e-8


# ------------------------------------------------------------ sizes and kernels

TILES = {16016, 16064, 64016, 64032, 64064, 128064, 128128, 256256}


def _tile(M, E, N, K, gate=0):
    f = dbs.lib().dbs_i8_tile
    f.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int] * 2
    return f(M, E, N, K, gate, 256)


def _parts(M, N, K):
    """The launches of a dense product."""
    f = dbs.lib().dbs_i8_part
    f.argtypes, f.restype = [ctypes.c_int64] * 3 + [ctypes.c_int], ctypes.c_int64
    n = f(M, N, K, 256)
    if n < 0:
        return [(M, -n, K), (M, N + n, K)]
    return [(n, N, K), (M - n, N, K)] if n < M else [(M, N, K)]


def test_dense_products_in_two_launches():
    assert all(len(_parts(*s)) == 1 for s in shapes.DENSE)
    parts = [_parts(*s) for s in shapes.PARTS]
    assert all(len(p) == 2 for p in parts)
    assert {p[0][0] < s[0] for p, s in zip(parts, shapes.PARTS)} == {True, False}
    rng = np.random.default_rng(6)
    for _ in range(3000):
        M, N, K = int(2 ** rng.uniform(0, 25)), int(2 ** rng.uniform(0, 21)), 16 * int(2 ** rng.uniform(0, 12.9))
        parts = _parts(M, N, K)
        assert sum(m * n for m, n, _ in parts) == M * N
        if len(parts) == 2:
            # whole tiles come first: what is behind them stays as aligned as the start
            (m, n, _), (m2, n2, _) = parts
            assert min(m, n, m2, n2) > 0 and ((m % 128 == 0 and n == N) or (n % 128 == 0 and m == M))


def test_gpu_sizes_reach_every_kernel():
    """The rule that the products go by puts the sizes of the GPU tests in every kernel."""
    assert {_tile(M, 1, N, K) for M, N, K in shapes.DENSE} == TILES
    assert {_tile(M, 1, N, K // 16 * 16) for M, N, K in shapes.POISON} >= TILES - {16016, 64016, 64032}
    ragged = {(tuple(s), N): _tile(sum(s), len(s), N, K) for s, N, K in shapes.RAGGED}
    assert set(ragged.values()) >= {16016, 16064, 64016, 64032}
    assert {_tile(M, E, N, K) for T, M, E, N, K in shapes.EXPERTS} | set(ragged.values()) == TILES
    gated = {_tile(M, E, 2 * N, K, 1) for T, M, E, N, K in shapes.EXPERTS}
    gated |= {_tile(sum(s), len(s), N, K, 1) for s, N, K in shapes.RAGGED}
    assert gated == TILES - {64016, 128064}
    # small tiles by several to a workgroup: more of them than workgroups
    for (sizes, N), tile in ragged.items():
        rows, cols = divmod(tile, 1000)
        if tile in (16016, 16064, 64016, 64032):
            tiles = sum(-(-n // rows) for n in sizes) * -(-N // cols)
            assert tiles > (512 if tile == 16016 else 256), (sizes, N, tile)


def test_the_rule_has_a_tile_for_every_size():
    rng = np.random.default_rng(5)
    for _ in range(2000):
        M, E = int(2 ** rng.uniform(0, 25)), int(2 ** rng.uniform(0, 10))
        N, K = 2 * int(2 ** rng.uniform(0, 20)), 16 * int(2 ** rng.uniform(0, 12.9))
        assert _tile(M, E, N, K) in TILES and _tile(M, E, N, K, 1) in TILES - {64016, 128064}
