"""Mixture-of-experts operators on the GPU against their plain 64-bit forms:
routing, the experts' products in every direction, the gate and the sums back
to tokens (-m gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _moe

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def _say(*a):
    print(*a, flush=True)


# ------------------------------------------------------------------ routing

def _logits(T, E, dtype, seed, closed=0.0):
    g = _gen(seed)
    x = torch.randn(T, E, generator=g)
    if closed:
        x[torch.rand(T, E, generator=g) < closed] = -float("inf")
        x[::5] = -float("inf")                       # tokens without any open expert
    return x.to(dtype)


ROUTE = [(1, 1, 1), (1, 64, 6), (1, 1024, 16), (3, 5, 5), (63, 17, 4), (64, 128, 8), (65, 128, 8), (257, 160, 6),
         (1000, 33, 2), (4100, 8, 2), (129, 1000, 16), (200, 512, 3)]


@pytest.mark.parametrize("T,E,k", ROUTE)
@pytest.mark.parametrize("dtype,renorm,closed", [(torch.float32, True, 0.0), (torch.bfloat16, False, 0.0),
                                                 (torch.float32, False, 0.5), (torch.bfloat16, True, 0.9)])
def test_route(T, E, k, dtype, renorm, closed):
    x = _logits(T, E, dtype, T * 1000 + E, closed)
    _say("route", T, E, k, dtype, renorm, closed)
    r = dbs.moe_route(x.cuda(), k, renormalize=renorm)
    experts, weights = _moe.route(_moe.f64(x), k, renorm)
    offsets, rows, slots = _moe.routing(experts, E)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    # the exponential's argument is rounded once (a step of its magnitude, at
    # most 20 here), E additions, a division
    assert np.all(np.abs(_moe.f64(r.weights) - weights) <= (E + 28) * 2.0 ** -23 * weights + 1e-30)


# both sides of the switch to three kernels (2048 tokens), experts over several
# workgroups of the column sums (16 each) and a rest, one to nine rows of counts a segment
MANY = [(2048, 33, 4), (2049, 33, 4), (2049, 16, 2), (4500, 160, 6), (4097, 17, 16), (2113, 600, 8), (2500, 1024, 3),
        (9000, 48, 8), (33000, 21, 2)]


@pytest.mark.parametrize("T,E,k", MANY)
@pytest.mark.parametrize("dtype,renorm,closed", [(torch.float32, True, 0.0), (torch.bfloat16, False, 0.6)])
def test_route_of_many_tokens(T, E, k, dtype, renorm, closed):
    x = _logits(T, E, dtype, T + 7 * E, closed)
    _say("route", T, E, k, dtype, renorm, closed)
    r = dbs.moe_route(x.cuda(), k, renormalize=renorm)
    experts, weights = _moe.route(_moe.f64(x), k, renorm)
    offsets, rows, slots = _moe.routing(experts, E)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    assert np.all(np.abs(_moe.f64(r.weights) - weights) <= (E + 28) * 2.0 ** -23 * weights + 1e-30)


def test_route_special_logits():
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    x = torch.tensor([[1.0, inf, inf, 0.0, -1.0],       # two infinities share
                      [nan, 1.0, nan, 2.0, -inf],       # two open experts
                      [low, low, low, low, low],        # the type's lowest value is a logit like any other
                      [low, 0.0, -inf, low, nan],
                      [nan, nan, nan, -inf, -inf],      # none open
                      [2.0, 2.0, 2.0, 2.0, 2.0],        # ties: the lower expert
                      [-inf, -inf, -inf, -inf, 3.0]])
    r = dbs.moe_route(x.cuda(), 3)
    assert r.experts.cpu().tolist() == [[1, 2, 0], [3, 1, -1], [0, 1, 2], [1, 0, 3], [-1, -1, -1], [0, 1, 2],
                                        [4, -1, -1]]
    w = r.weights.cpu()
    assert w[0].tolist() == [0.5, 0.5, 0.0]
    assert torch.allclose(w[2], torch.full((3,), 1 / 3)) and w[3].tolist() == [1.0, 0.0, 0.0]
    assert w[4].tolist() == [0.0, 0.0, 0.0] and w[6].tolist() == [1.0, 0.0, 0.0]
    total = int(r.offsets[-1])
    assert total == 3 + 2 + 3 + 3 + 0 + 3 + 1
    assert r.rows[total:].eq(-1).all() and r.rows[:total].ge(0).all()
    d = torch.randn(7, 3, generator=_gen(3))
    got = _moe.f64(dbs.moe_route_backward(x.cuda(), r.experts, d.cuda()))
    want = _moe.route_grad(_moe.f64(x), r.experts.cpu().numpy(), _moe.f64(d), True)
    assert np.all(np.isfinite(got)) and np.allclose(got, want, rtol=0, atol=40 * 2.0 ** -23 * float(d.abs().max()))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (33, 160, 6), (100, 17, 4), (17, 1024, 16), (50, 300, 8)])
@pytest.mark.parametrize("dtype,renorm,closed", [(torch.float32, True, 0.0), (torch.bfloat16, False, 0.0),
                                                 (torch.float32, False, 0.6), (torch.bfloat16, True, 0.8)])
def test_route_backward(T, E, k, dtype, renorm, closed):
    x = _logits(T, E, dtype, T + E, closed)
    d = torch.randn(T, k, generator=_gen(5))
    experts, _ = _moe.route(_moe.f64(x), k, renorm)
    got = _moe.f64(dbs.moe_route_backward(x.cuda(), torch.tensor(experts, dtype=torch.int32).cuda(), d.cuda(),
                                          renormalize=renorm))
    want = _moe.route_grad(_moe.f64(x), experts, _moe.f64(d), renorm)
    # p to (E + 28) steps as above, the inner sum over E terms of at most |d|
    bound = (2 * E + 60) * 2.0 ** -23 * float(d.abs().max())
    if dtype == torch.bfloat16:
        bound = bound + _moe.HALF_STEP * np.abs(want)
    assert np.all(np.abs(got - want) <= bound)


def test_route_gradient_against_differences():
    T, E, k, h = 6, 12, 3, 2.0 ** -7
    x = torch.randn(T, E, generator=_gen(11))
    d = torch.randn(T, k, generator=_gen(12))
    for renorm in (True, False):
        r = dbs.moe_route(x.cuda(), k, renormalize=renorm)
        g = _moe.f64(dbs.moe_route_backward(x.cuda(), r.experts, d.cuda(), renormalize=renorm))
        experts = r.experts.cpu()
        for t in range(T):
            for e in range(E):
                ends = []
                for s in (h, -h):
                    y = x.clone()
                    y[t, e] += s
                    q = dbs.moe_route(y.cuda(), k, renormalize=renorm)
                    if not torch.equal(q.experts.cpu(), experts):
                        break                     # the choice changes here: no derivative
                    ends.append(float((q.weights.cpu().double() * d.double()).sum()))
                if len(ends) == 2:
                    # differences: h^2 / 6 of the third derivative (at most 1 times sum |d|), rounding / h
                    tol = float(d[t].abs().sum()) * (h * h + 64 * 2.0 ** -23 * T / h)
                    assert abs((ends[0] - ends[1]) / (2 * h) - g[t, e]) <= tol


def test_route_repeats_and_runs_on_the_callers_stream():
    x = _logits(3000, 96, torch.float32, 9).cuda()
    a = dbs.moe_route(x, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = dbs.moe_route(x, 6)
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)


# ----------------------------------------------------------------- products

def _groups(kind, E, M, seed):
    """Ascending offsets of E groups over at most M rows."""
    rng = np.random.default_rng(seed)
    if kind == "even":
        return np.array([M * e // E for e in range(E + 1)])
    if kind == "one":                       # everything to one expert
        return np.array([0] * (E // 2 + 1) + [M] * (E - E // 2))
    if kind == "none":                      # no expert has a row
        return np.zeros(E + 1, dtype=int)
    if kind == "short":                     # rows are left over behind the last group
        return np.sort(np.concatenate([[0], rng.integers(0, max(1, M * 2 // 3), E)]))
    cuts = np.sort(rng.integers(0, M + 1, E - 1)) if E > 1 else np.array([], dtype=int)
    return np.concatenate([[0], cuts, [M]])


# T, M (None: sorted already), E, N, K, groups
SHAPES = [
    (1, 8, 64, 64, 256, "ragged"), (1, 1, 1, 1, 8, "even"), (5, 7, 3, 33, 40, "ragged"),
    (48, 384, 128, 96, 200, "ragged"), (300, 700, 4, 264, 136, "ragged"), (64, 129, 2, 257, 64, "even"),
    (900, 1800, 8, 520, 320, "ragged"), (2000, 2050, 2, 300, 72, "one"), (513, None, 3, 256, 128, "even"),
    (33, None, 5, 130, 8, "short"), (400, 900, 7, 144, 104, "short"), (16, 40, 6, 72, 64, "none"),
    (700, 1500, 5, 776, 1032, "ragged"), (20, 60, 1000, 40, 64, "ragged"),
]


# rows and columns enough for the 256-row tiles: rests of one to four blocks,
# column starts past 2048, one to a few stages, no whole pieces
LARGE = [
    (600, 3000, 5, 4360, 136, "ragged"), (2000, 6000, 3, 2304, 200, "ragged"),
    (5000, None, 40, 1032, 264, "ragged"), (64000, None, 3, 97, 40, "ragged"), (64500, None, 2, 72, 8, "one"),
    (9000, None, 6, 2312, 104, "none"), (4000, 9000, 7, 2312, 328, "short"), (300, 4097, 1, 4099, 64, "even"),
    (1, 2600, 2, 4104, 128, "even"),
]


# for the 128-row tiles
MID = [
    (900, 2048, 2, 2056, 200, "ragged"), (500, 4000, 8, 1032, 40, "ragged"), (4000, None, 1, 1033, 264, "even"),
    (8200, None, 5, 608, 328, "ragged"), (1300, 1300, 2, 4360, 72, "ragged"), (3800, None, 3, 1352, 136, "short"),
    (1200, None, 3, 4096, 104, "ragged"), (700, 8300, 5, 600, 72, "ragged"), (2900, None, 2, 1544, 328, "ragged"),
]
HALF = [(T, M, E, N // 2, K, groups) for T, M, E, N, K, groups in MID]      # the same behind the gate


def test_shapes_reach_every_tile_height():
    """The rule of moe.cpp on 256 CUs: LARGE goes to 256-row tiles and MID to
    128-row tiles of a K-major product, and in every form the shapes of the tests
    reach every height three times at least."""
    def height(M, E, N, mn, gate):
        cols, met = N // 2 if gate else N, min(M, -(-2 * M * E // (2 * M + E)))
        per_cu = lambda tm, tn: max(M // tm + met // 2, met) * -(-cols // tn) / 256
        w = met * N / 65536

        def rounds(tm, stage):
            n = per_cu(tm, 128 if gate else 256)
            return n // 1 * max(stage, w / n) + (stage if n % 1 else 0.0)
        small = max((0.39 if mn else 0.22) * per_cu(64, 128 if mn else 32 if gate else 64), 1.1 * w)
        mid, large = rounds(128, 0.85), rounds(256, 1.0)
        return 64 if small <= mid and small <= large else 128 if mid < large else 256
    for shapes, want in ((LARGE, 256), (MID, 128)):
        for T, M, E, N, K, groups in shapes:
            assert height(M or T, E, N, False, False) == want, (T, M, E, N, K, groups)
    for mn, gate in ((False, False), (False, True), (True, False)):
        reached = [height(M or T, E, 2 * N if gate else N, mn, gate)
                   for T, M, E, N, K, _ in SHAPES + MID + LARGE + (HALF if gate else []) if not mn or N % 8 == 0]
        assert all(reached.count(h) >= 3 for h in (64, 128, 256)), (mn, gate, reached)


def test_dw_shapes_reach_both_tiles():
    """As above, for the rule of moe_dw on the groups that test_dw makes."""
    def small(off, N, K, accumulate, f32):
        rows = np.diff(off)
        rows = rows[rows > 0] if accumulate else rows
        stages = -(-rows // 64)
        few, many = -(-N // 64) * -(-K // 128), -(-N // 256) * -(-K // 256)
        wgs, n = min(256, (len(off) - 1) * few), len(rows)
        longest = stages.max(initial=0)
        large = (90 if f32 else 50) * np.ceil(many * n / wgs) + max(
            13 * longest, 16 * many * np.maximum(stages, 2).sum() / wgs)
        return 10 * np.ceil(few * n / wgs) + max(3.5 * longest, 5 * few * np.maximum(stages, 4).sum() / wgs) < large
    for shapes, want in ((NARROW, True), (WIDE, False)):
        for T, M, E, N, K, groups in shapes:
            assert small(_groups(groups, E, M or T, N + K + 3), N, K, False, False) == want, (T, M, E, N, K, groups)


def _case(T, M, E, K, groups, seed):
    g = _gen(seed)
    X = _bf16(g, T, K)
    off = _groups(groups, E, M or T, seed)
    rows = None
    if M is not None:
        rows = torch.randint(0, T, (M,), generator=g, dtype=torch.int32)
    return g, X, off, rows


def _gpu(X, off, rows):
    return X.cuda(), torch.tensor(off, dtype=torch.int32).cuda(), None if rows is None else rows.cuda()


@pytest.mark.parametrize("T,M,E,N,K,groups", SHAPES + MID + LARGE)
def test_product(T, M, E, N, K, groups):
    g, X, off, rows = _case(T, M, E, K, groups, N + K)
    W = _bf16(g, E, N, K)
    _say("product", T, M, E, N, K, groups)
    x, o, r = _gpu(X, off, rows)
    out = torch.full((M or T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = _moe.f64(dbs.gemm_moe_bf16(x, W.cuda(), o, r, out=out))
    D, S = _moe.product(_moe.f64(X), _moe.f64(W), off, None if rows is None else rows.numpy(), False)
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K))
    assert np.all(got[off[-1]:] == 0)


@pytest.mark.parametrize("T,M,E,N,K,groups", [s for s in SHAPES + MID + LARGE if s[3] % 8 == 0])
def test_product_transposed(T, M, E, N, K, groups):
    g, X, off, rows = _case(T, M, E, K, groups, N + K + 1)
    W = _bf16(g, E, K, N)
    _say("transposed", T, M, E, N, K, groups)
    x, o, r = _gpu(X, off, rows)
    got = _moe.f64(dbs.gemm_moe_bf16(x, W.cuda(), o, r, lw=dbs.MN_MAJOR))
    D, S = _moe.product(_moe.f64(X), _moe.f64(W), off, None if rows is None else rows.numpy(), True)
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K))
    assert np.all(got[off[-1]:] == 0)


@pytest.mark.parametrize("T,M,E,F,K,groups", SHAPES + MID + LARGE + HALF)
def test_product_gated(T, M, E, F, K, groups):
    g, X, off, rows = _case(T, M, E, K, groups, F + K + 2)
    W = _bf16(g, E, 2 * F, K, scale=K ** -0.5 * 2)
    _say("gated", T, M, E, F, K, groups)
    x, o, r = _gpu(X, off, rows)
    got = _moe.f64(dbs.gemm_moe_swiglu_bf16(x, W.cuda(), o, r))
    D, S = _moe.product(_moe.f64(X), _moe.f64(W), off, None if rows is None else rows.numpy(), False)
    acc = K * 2.0 ** -23 * S
    a, u = D[:, :F], D[:, F:]
    assert np.all(np.abs(got - _moe.silu(a) * u) <= _moe.gate_bound(a, u, acc[:, :F], acc[:, F:]))


# few or thin matrices under many rows: one to several of the smaller dw tiles
# per workgroup, groups that end in a stage or have none
NARROW = [
    (300, 192, 1, 8, 8, "even"), (300, 193, 1, 72, 136, "even"), (100, 4000, 4, 64, 128, "ragged"),
    (2000, 2000, 5, 200, 264, "short"), (500, 3000, 3, 48, 1032, "one"), (700, 2400, 12, 264, 648, "none"),
    (4000, None, 12, 136, 520, "ragged"), (1030, None, 5, 56, 1160, "ragged"), (900, 12000, 60, 56, 1544, "ragged"),
    (700, 10000, 50, 320, 640, "ragged"), (64, 13000, 60, 320, 392, "one"), (700, 3000, 6, 1032, 1288, "ragged"),
    (3000, None, 6, 1032, 1288, "one"),
]
# the larger ones: long groups, several tiles per workgroup, a stage or two per group
WIDE = [
    (5000, None, 40, 1032, 264, "ragged"), (150, 2600, 21, 1040, 648, "short"), (200, 1300, 130, 520, 264, "ragged"),
    (700, 5200, 4, 1032, 2056, "even"), (5200, None, 4, 1032, 2056, "even"),
]


@pytest.mark.parametrize("T,M,E,N,K,groups", [s for s in SHAPES if s[3] % 8 == 0] + NARROW + WIDE)
@pytest.mark.parametrize("out", ["bf16", "f32", "add"])
def test_dw(T, M, E, N, K, groups, out):
    g, X, off, rows = _case(T, M, E, K, groups, N + K + 3)
    dY = _bf16(g, M or T, N)
    _say("dw", T, M, E, N, K, groups, out)
    x, o, r = _gpu(X, off, rows)
    D, S = _moe.dw(_moe.f64(dY), _moe.f64(X), off, None if rows is None else rows.numpy())
    n = int(np.diff(off).max())
    acc = (n + 1) * 2.0 ** -23 * S
    if out == "bf16":
        got = _moe.f64(dbs.gemm_moe_dw_bf16(dY.cuda(), x, o, r))
        assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, n))
    elif out == "f32":
        got = _moe.f64(dbs.gemm_moe_dw_bf16(dY.cuda(), x, o, r, out_dtype=torch.float32))
        assert np.all(np.abs(got - D) <= acc)
    else:
        base = torch.randn(E, N, K, generator=g)
        got = dbs.gemm_moe_dw_bf16(dY.cuda(), x, o, r, out=base.cuda(), accumulate=True)
        b = _moe.f64(base)
        assert np.all(np.abs(_moe.f64(got) - (b + D)) <= acc + 2.0 ** -23 * (np.abs(b) + np.abs(D)))


@pytest.mark.parametrize("rows_of_masked", ["inf", "nan"])
def test_values_outside_a_group_stay_outside(rows_of_masked):
    """Infinities and NaN in rows that no expert takes, in other experts'
    matrices and behind K reach nothing."""
    bad = float(rows_of_masked)
    T, E, N, K = 40, 4, 72, 40
    g = _gen(21)
    X, W = _bf16(g, T, K), _bf16(g, E, N, K)
    off = np.array([0, 10, 10, 25, 30])
    X[30:] = bad                         # behind the last group
    W[1] = bad                           # an expert without rows
    x, o, _ = _gpu(X, off, None)
    Xc = _moe.f64(X)
    Xc[30:] = 0
    Wc = _moe.f64(W)
    Wc[1] = 0
    D, S = _moe.product(Xc, Wc, off, None, False)
    got = _moe.f64(dbs.gemm_moe_bf16(x, W.cuda(), o))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K)) and np.all(got[30:] == 0)
    wt = W.transpose(1, 2).contiguous().cuda()
    got = _moe.f64(dbs.gemm_moe_bf16(x, wt, o, lw=dbs.MN_MAJOR))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K))
    dY = _bf16(g, T, N)
    dY[30:] = bad
    dYc = _moe.f64(dY)
    dYc[30:] = 0
    D, S = _moe.dw(dYc, Xc, off, None)
    got = _moe.f64(dbs.gemm_moe_dw_bf16(dY.cuda(), x, o))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, 15))
    # one token's NaN stays in its rows
    X2 = _bf16(g, T, K)
    X2[7] = bad
    rows = torch.randint(0, T, (T,), generator=g, dtype=torch.int32)
    got = _moe.f64(dbs.gemm_moe_bf16(X2.cuda(), _bf16(g, E, N, K).cuda(), o, rows.cuda()))
    assert np.all(np.isfinite(got[:30][rows[:30].numpy() != 7]))


def test_row_indices_outside_x_are_zero_rows():
    g = _gen(31)
    T, E, N, K = 20, 2, 64, 64
    X, W, dY = _bf16(g, T, K), _bf16(g, E, N, K), _bf16(g, 30, N)
    rows = torch.randint(0, T, (30,), generator=g, dtype=torch.int32)
    rows[3], rows[17] = -1, T
    off = np.array([0, 12, 30])
    x, o, r = _gpu(X, off, rows)
    D, S = _moe.product(_moe.f64(X), _moe.f64(W), off, rows.numpy(), False)
    got = _moe.f64(dbs.gemm_moe_bf16(x, W.cuda(), o, r))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K)) and np.all(got[[3, 17]] == 0)
    D, S = _moe.dw(_moe.f64(dY), _moe.f64(X), off, rows.numpy())
    got = _moe.f64(dbs.gemm_moe_dw_bf16(dY.cuda(), x, o, r))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, 30))


def test_large_tiles_keep_foreign_rows_out():
    """Infinities behind the last group, in an expert without rows and in rows
    of X that no index names; indices outside X."""
    g = _gen(33)
    T, E, N, K = 700, 3, 4360, 136
    off = np.array([0, 1201, 1201, 2600])
    M, bad = 3000, float("inf")
    X, W = _bf16(g, T, K), _bf16(g, E, N, K)
    rows = torch.randint(0, T - 1, (M,), generator=g, dtype=torch.int32)
    rows[5], rows[1200], rows[1201], rows[2599] = -1, T, 1 << 30, -(1 << 31)
    X[T - 1], W[1] = bad, bad
    rows[2600:] = T - 1
    Xc, Wc = _moe.f64(X), _moe.f64(W)
    Xc[T - 1], Wc[1] = 0, 0
    x, o, r = _gpu(X, off, rows)
    D, S = _moe.product(Xc, Wc, off, rows.numpy(), False)
    got = _moe.f64(dbs.gemm_moe_bf16(x, W.cuda(), o, r))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K))
    assert np.all(got[2600:] == 0) and np.all(got[[5, 1200, 1201, 2599]] == 0)
    got = _moe.f64(dbs.gemm_moe_bf16(x, W.transpose(1, 2).contiguous().cuda(), o, r, lw=dbs.MN_MAJOR))
    assert np.all(np.abs(got - D) <= _moe.product_bound(D, S, K)) and np.all(got[2600:] == 0)
    a, u, acc = D[:, :N // 2], D[:, N // 2:], K * 2.0 ** -23 * S
    got = _moe.f64(dbs.gemm_moe_swiglu_bf16(x, W.cuda(), o, r))
    assert np.all(np.abs(got - _moe.silu(a) * u) <= _moe.gate_bound(a, u, acc[:, :N // 2], acc[:, N // 2:]))
    assert np.all(got[2600:] == 0)


def test_dw_against_differences():
    """d/dW of L = sum C * (X W^T) is C^T X; L is linear in W, so its
    differences hold it to rounding, with integers exactly."""
    g = _gen(41)
    T, E, N, K = 24, 3, 16, 16
    X = torch.randint(-3, 4, (T, K), generator=g).to(torch.bfloat16)
    W = torch.randint(-3, 4, (E, N, K), generator=g).to(torch.bfloat16)
    C = torch.randint(-3, 4, (T, N), generator=g).to(torch.bfloat16)
    o = torch.tensor([0, 9, 9, 24], dtype=torch.int32).cuda()
    d = dbs.gemm_moe_dw_bf16(C.cuda(), X.cuda(), o, out_dtype=torch.float32).cpu()
    loss = lambda w: float((dbs.gemm_moe_bf16(X.cuda(), w.cuda(), o).cpu().double() * C.double()).sum())
    base = loss(W)
    for e, n, k in [(0, 0, 0), (0, 15, 3), (1, 4, 4), (2, 7, 15), (2, 0, 8)]:
        V = W.clone()
        V[e, n, k] += 1
        assert loss(V) - base == float(d[e, n, k])
    # and with respect to the rows
    dx = dbs.gemm_moe_bf16(C.cuda(), W.cuda(), o, lw=dbs.MN_MAJOR).cpu()
    loss_x = lambda x: float((dbs.gemm_moe_bf16(x.cuda(), W.cuda(), o).cpu().double() * C.double()).sum())
    for t, k in [(0, 0), (8, 5), (9, 15), (23, 1)]:
        Z = X.clone()
        Z[t, k] += 1
        assert loss_x(Z) - base == float(dx[t, k])


# -------------------------------------------------------------- gate, sums

@pytest.mark.parametrize("M,F", [(1, 1), (1, 8), (3, 7), (5, 264), (1000, 40), (77, 1416), (2, 4099)])
def test_swiglu(M, F):
    g = _gen(M + F)
    H, dA = _bf16(g, M, 2 * F, scale=4.0), _bf16(g, M, F)
    H[0, 0] = -300.0                          # the exponential overflows: silu is 0
    a, u, d = _moe.f64(H[:, :F]), _moe.f64(H[:, F:]), _moe.f64(dA)
    got = _moe.f64(dbs.swiglu(H.cuda()))
    assert np.all(np.abs(got - _moe.silu(a) * u) <= _moe.gate_bound(a, u, 0.0, 0.0))
    got = _moe.f64(dbs.swiglu_backward(dA.cuda(), H.cuda()))
    s = 1 / (1 + np.exp(-a))
    da, du = d * u * s * (1 + a * (1 - s)), d * a * s
    # steps as in gate_bound; 1 + g (1 - s) loses what its terms' magnitudes hold
    rel = (16 + np.abs(a)) * 2.0 ** -22
    slack = rel * np.abs(d * u * s) * (1 + np.abs(a) * (1 - s) * (1 + np.abs(a)))
    assert np.all(np.abs(got[:, :F] - da) <= slack + _moe.HALF_STEP * (np.abs(da) + slack) + _moe.TINY)
    assert np.all(np.abs(got[:, F:] - du) <= (rel + _moe.HALF_STEP * (1 + rel)) * np.abs(du) + _moe.TINY)


def _far_below():
    """Gates where e^-g leaves fp32's normal range or fp32, and what they meet:
    silu(g) u is a normal number for some of them."""
    g = torch.arange(-120, -70, 0.5)
    u = torch.tensor([1.0, -3.0, 2.0 ** 40, -2.0 ** 100])
    return g.repeat(4).to(torch.bfloat16), u.repeat_interleave(len(g)).to(torch.bfloat16)


def test_swiglu_far_below_zero():
    g, u = _far_below()
    a, b = _moe.f64(g), _moe.f64(u)
    H = torch.cat([g, u]).view(1, -1)
    got = _moe.f64(dbs.swiglu(H.cuda()))[0]
    assert np.all(np.abs(got - _moe.silu(a) * b) <= _moe.gate_bound(a, b, 0.0, 0.0))
    d = torch.tensor([0.75, -2.0]).repeat(len(g) // 2).to(torch.bfloat16)
    got = _moe.f64(dbs.swiglu_backward(d.view(1, -1).cuda(), H.cuda()))[0]
    dd, s = _moe.f64(d), 1 / (1 + np.exp(-a))
    da, du = dd * b * s * (1 + a * (1 - s)), dd * a * s
    # (bounds of test_swiglu)
    rel = (16 + np.abs(a)) * 2.0 ** -22
    slack = rel * np.abs(dd * b * s) * (1 + np.abs(a) * (1 - s) * (1 + np.abs(a)))
    assert np.all(np.abs(got[:len(a)] - da) <= slack + _moe.HALF_STEP * (np.abs(da) + slack) + _moe.TINY)
    assert np.all(np.abs(got[len(a):] - du) <= (rel + _moe.HALF_STEP * (1 + rel)) * np.abs(du) + _moe.TINY)


@pytest.mark.parametrize("M", [1, 200, 60000])
def test_product_gated_far_below_zero(M):
    """The same out of the product's registers: one term per sum."""
    g, u = _far_below()
    a, b = _moe.f64(g), _moe.f64(u)
    F = len(g)
    X, W = torch.zeros(M, 8, dtype=torch.bfloat16), torch.zeros(1, 2 * F, 8, dtype=torch.bfloat16)
    X[:, 3] = 1.0
    W[0, :, 3] = torch.cat([g, u])
    got = dbs.gemm_moe_swiglu_bf16(X.cuda(), W.cuda(), torch.tensor([0, M], dtype=torch.int32).cuda())
    first = _moe.f64(got[0])
    assert np.all(np.abs(first - _moe.silu(a) * b) <= _moe.gate_bound(a, b, 0.0, 0.0))
    assert bool((got == got[0]).all())


def test_swiglu_gradient_against_differences():
    g = _gen(51)
    M, F, h = 3, 8, 0.5
    H = (torch.randint(-8, 9, (M, 2 * F), generator=g) / 4).to(torch.bfloat16)
    one = torch.ones(M, F, dtype=torch.bfloat16)
    got = _moe.f64(dbs.swiglu_backward(one.cuda(), H.cuda()))
    hi, lo = H.clone(), H.clone()
    hi[:, F:] += h
    lo[:, F:] -= h                            # linear in the up half: only rounding is left
    d = (_moe.f64(dbs.swiglu(hi.cuda())) - _moe.f64(dbs.swiglu(lo.cuda()))) / (2 * h)
    assert np.all(np.abs(d - got[:, F:]) <= 4 * _moe.HALF_STEP * 3.0 / h)
    hi, lo = H.clone(), H.clone()
    hi[:, :F] += h
    lo[:, :F] -= h
    d = (_moe.f64(dbs.swiglu(hi.cuda())) - _moe.f64(dbs.swiglu(lo.cuda()))) / (2 * h)
    # h^2 / 6 of silu's third derivative (below 0.5), |u| <= 2, and rounding
    assert np.all(np.abs(d - got[:, :F]) <= h * h / 6 * 0.5 * 2 + 4 * _moe.HALF_STEP * 5.0 / h)


def _slots(T, k, drop, seed):
    g = _gen(seed)
    E = 4
    experts = torch.randint(0, E, (T, k), generator=g)
    if drop:
        experts[torch.rand(T, k, generator=g) < drop] = -1
        experts[:1] = -1
    offsets, rows, slots = _moe.routing(experts.numpy(), E)
    return offsets, slots


@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 4096), (3, 2, 7), (37, 6, 264), (200, 16, 33), (129, 4, 1032)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_combine(T, k, H, drop):
    g = _gen(T + H)
    offsets, slots = _slots(T, k, drop, T)
    Y, dO, w = _bf16(g, T * k, H), _bf16(g, T, H), torch.rand(T, k, generator=g)
    bad = Y.clone()
    bad[offsets[-1]:] = float("nan")                 # rows of no pair are not read
    s = torch.tensor(slots, dtype=torch.int32).cuda()
    taken = slots >= 0
    y = _moe.f64(Y)[np.where(taken, slots, 0)] * taken[..., None]
    for weights in (w, None):
        ww = np.ones((T, k)) if weights is None else _moe.f64(w)
        want = (ww[..., None] * y).sum(1)
        size = (ww[..., None] * np.abs(y)).sum(1)
        got = _moe.f64(dbs.moe_combine(bad.cuda(), s, None if weights is None else weights.cuda()))
        assert np.all(np.abs(got - want) <= _moe.product_bound(want, size, 2 * k))
    o = torch.tensor(offsets, dtype=torch.int32).cuda()
    dY, dw = dbs.moe_combine_backward(dO.cuda(), bad.cuda(), s, w.cuda(), o)
    d = _moe.f64(dO)
    want = (d[:, None] * y).sum(-1)
    size = (np.abs(d)[:, None] * np.abs(y)).sum(-1)
    assert np.all(np.abs(_moe.f64(dw) - want) <= (H + 1) * 2.0 ** -23 * size)
    wantY = np.zeros((T * k, H))
    for t, j in zip(*np.nonzero(taken)):
        wantY[slots[t, j]] = _moe.f64(w)[t, j] * d[t]
    got = _moe.f64(dY)
    assert np.all(np.abs(got - wantY) <= _moe.HALF_STEP * (1 + 2.0 ** -22) * np.abs(wantY) + _moe.TINY)
    assert np.all(got[offsets[-1]:] == 0)


def test_arrays_off_16_byte_addresses():
    """Row lengths of whole pieces whose base address is not one."""
    g = _gen(61)
    flat = _bf16(g, 1 + 6 * 32).cuda()
    H = flat[1:].view(6, 32)
    a, u = _moe.f64(H[:, :16]), _moe.f64(H[:, 16:])
    assert np.all(np.abs(_moe.f64(dbs.swiglu(H)) - _moe.silu(a) * u) <= _moe.gate_bound(a, u, 0.0, 0.0))
    s = torch.tensor([[0, 3], [5, -1]], dtype=torch.int32).cuda()
    got = _moe.f64(dbs.moe_combine(H, s))
    y = _moe.f64(H)
    want = np.stack([y[0] + y[3], y[5]])
    assert np.all(np.abs(got - want) <= _moe.product_bound(want, np.abs(want) + 8, 2))
