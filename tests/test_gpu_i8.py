"""8-bit integer operators on the GPU against their plain 64-bit forms (-m gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _i8, _moe

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _codes(g, *shape):
    """Every code from -128 on."""
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int8)


def _scales(g, *shape):
    return torch.exp2(torch.rand(*shape, generator=g) * 8 - 10)


def _say(*a):
    print(*a, flush=True)


# ------------------------------------------------------------- the quantiser

# both sides of every size of row a kernel holds, whole pieces and not
QUANT = [(1, 1), (3, 7), (1, 16), (5, 8), (64, 512), (9, 520), (7, 1024), (6, 1032), (5, 2048), (4, 2056), (3, 4096),
         (2, 4104), (3, 8192), (2, 8200), (2, 16384), (2, 16392), (1, 40000), (2, 2049), (1, 4101), (1000, 48), (257, 100),
         (4097, 520), (4096, 1024), (16385, 1032)]


@pytest.mark.parametrize("M,K", QUANT)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant(M, K, dtype):
    g = _gen(M * 100003 + K)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-40, 40, (M, 1), generator=g).float())).to(dtype)
    _say("quant", M, K, dtype)
    q, s = dbs.quant_i8(x.cuda())
    codes, scales = _i8.quant(_moe.f64(x))
    assert np.array_equal(q.cpu().numpy(), codes)
    assert np.all(np.abs(_moe.f64(s) - scales) <= _i8.HALF_F32 * scales)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quant_next_to_ties(dtype):
    """Rows whose quotients lie on ties and within a last place of them."""
    rows = []
    for amax in (127.0, 254.0, 2.0, 1.0, 3.0, 100.0, 0.75, 96.0):
        ties = (np.arange(127) + 0.5) * amax / 127
        near = np.concatenate([ties, np.nextafter(ties.astype(np.float32), np.float32(np.inf)),
                               np.nextafter(ties.astype(np.float32), np.float32(0))]).astype(np.float32)
        rows.append(np.concatenate([near, -near, [amax], np.zeros(768 - 2 * len(near) - 1)]).astype(np.float32))
    x = torch.tensor(np.array(rows)).to(dtype)
    q, _ = dbs.quant_i8(x.cuda())
    assert np.array_equal(q.cpu().numpy(), _i8.quant(_moe.f64(x))[0])


@pytest.mark.parametrize("K", [24, 25, 5000])
def test_quant_special_rows(K):
    g = _gen(K)
    x = torch.randn(9, K, generator=g)
    x[0] = 0
    x[1] *= 1e-43                                        # subnormal
    x[2] = torch.where(x[2] > 0, 3.3e38, -3.4e38)
    x[3, K - 1] = float("inf")
    x[4, 0] = float("nan")
    x[5] = 1e-45
    x[6] *= 2.0 ** -101
    x[7, 1] = -float("inf")
    q, s = dbs.quant_i8(x.cuda())
    codes, scales = _i8.quant(_moe.f64(x))
    assert np.array_equal(q.cpu().numpy(), codes)
    assert torch.isnan(s[[3, 4, 7]]).all() and float(s[0]) == 0 and not q[0].any()
    fine = [0, 1, 2, 5, 6, 8]
    assert np.all(np.abs(_moe.f64(s)[fine] - scales[fine]) <= _i8.HALF_F32 * scales[fine] + 2.0 ** -150)


def test_quant_rows_on_odd_addresses():
    """Rows of a tensor that starts two (four) bytes into its storage."""
    g = _gen(4)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn(1 + 6 * 64, generator=g).to(dtype).cuda()[1:].view(6, 64)
        q, s = dbs.quant_i8(x)
        codes, scales = _i8.quant(_moe.f64(x))
        assert np.array_equal(q.cpu().numpy(), codes)


# ---------------------------------------------------------- the dense product

# one row to several tiles, every number of 64-row blocks, widths and depths that
# end inside a tile (a vector, a stage), every tile, few and many stages
DENSE = [(1, 1, 16), (1, 64, 128), (1, 8192, 4096), (2, 33, 48), (5, 100, 144), (16, 256, 1024), (17, 1000, 2064),
         (48, 4096, 512), (63, 65, 912), (64, 2050, 1040), (65, 64, 16), (100, 300, 3200), (200, 4097, 272),
         (256, 256, 384), (300, 520, 4096), (513, 2047, 528), (1024, 1024, 1024), (700, 8200, 256), (2047, 4102, 400),
         (4096, 4100, 128), (8192, 513, 160), (64, 8170, 528), (512, 8170, 512), (1030, 4099, 784),
         (1030, 8170, 784), (2157, 6150, 1040), (2500, 4099, 1040),
         (16, 8200, 2064), (3, 20000, 528), (13, 17002, 400)]

# in two launches, the second for the last rows or the last columns
PARTS = [(1679, 2389, 2144), (2196, 1902, 3248), (330, 10932, 2208), (3104, 1298, 2848), (992, 4108, 2320)]


@pytest.mark.parametrize("M,N,K", DENSE + PARTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(M, N, K, dtype):
    g = _gen(M * 7 + N * 11 + K)
    A, B, sA, sB = _codes(g, M, K), _codes(g, N, K), _scales(g, M), _scales(g, N)
    _say("gemm", M, N, K, dtype)
    D = dbs.gemm_i8(A.cuda(), sA.cuda(), B.cuda(), sB.cuda(), out_dtype=dtype)
    want = _i8.product(*(_moe.f64(t) for t in (A, sA, B, sB)))
    assert D.dtype == dtype
    assert np.all(np.abs(_moe.f64(D) - want) <= _i8.product_bound(want, dtype == torch.bfloat16))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gemm_sums_are_whole_at_the_largest_k(M):
    """131056 products of -128 and -128, and of +-127: the sums are exact and do not leave 32 bits."""
    K, N = 131056, 80
    A = torch.full((M, K), -128, dtype=torch.int8)
    B = torch.full((N, K), -128, dtype=torch.int8)
    B[1::2] = 127
    B[2] = _codes(_gen(1), K)
    one = torch.ones(max(M, N)).cuda()
    D = dbs.gemm_i8(A.cuda(), one[:M], B.cuda(), one[:N], out_dtype=torch.float32).cpu()
    want = (A[:1].double() @ B.double().t()).float()
    assert torch.equal(D, want.expand(M, N))


def test_gemm_out_and_values():
    g = _gen(9)
    A, B, sA, sB = (t.cuda() for t in (_codes(g, 70, 64), _codes(g, 90, 64), _scales(g, 70), _scales(g, 90)))
    want = dbs.gemm_i8(A, sA, B, sB)
    out = torch.full((70, 90), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert dbs.gemm_i8(A, sA, B, sB, out=out) is out and torch.equal(out, want)
    # a NaN scale is in its row alone, one of B in its column alone; a zero scale gives zeros
    sA[3], sB[5], sA[4] = float("nan"), float("nan"), 0.0
    D = dbs.gemm_i8(A, sA, B, sB)
    bad = torch.zeros(70, 90, dtype=torch.bool, device="cuda")
    bad[3], bad[:, 5] = True, True
    assert torch.equal(torch.isnan(D), bad) and bool((D[4][~bad[4]] == 0).all())
    keep = ~bad
    keep[4] = False
    assert torch.equal(D[keep], want[keep])
    # an output on an odd address, behind which nothing is written
    store = torch.full((70 * 90 + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    odd = store[1:1 + 70 * 90].view(70, 90)
    dbs.gemm_i8(A, torch.ones_like(sA), B, torch.ones_like(sB), out=odd)
    assert torch.equal(odd, dbs.gemm_i8(A, torch.ones_like(sA), B, torch.ones_like(sB)))
    assert store[0] == 7 and bool((store[-2:] == 7).all())


# -------------------------------------------------------- the experts' product


def _split(M, E, seed, first=0, last=0):
    """Offsets of E groups over rows first .. M - last - 1, some empty."""
    rng = np.random.default_rng(seed)
    w = rng.exponential(size=E) * (rng.random(E) > 0.3)
    w = w / max(w.sum(), 1e-9)
    cut = np.round(np.cumsum(w) * (M - first - last)).astype(int) + first
    cut[-1] = M - last if w.sum() > 0 else first
    return np.concatenate([[first], np.maximum.accumulate(cut)])


# T, M, E, N, K: gathered rows; sorted ones where T == M
EXPERTS = [(1, 2, 4, 64, 128), (3, 9, 5, 33, 48), (7, 7, 1, 100, 16), (16, 64, 64, 130, 272), (48, 384, 128, 96, 512),
           (100, 600, 8, 513, 1040), (300, 900, 3, 264, 400), (500, 500, 40, 1000, 96), (600, 2400, 4, 1030, 160),
           (2000, 8000, 12, 520, 256), (4099, 4099, 6, 2050, 144), (40, 200, 1024, 40, 80),
           (3000, 9000, 6, 2050, 528), (300, 1500, 6, 1030, 800), (300, 250, 1, 8000, 1040)]


@pytest.mark.parametrize("T,M,E,N,K", EXPERTS)
@pytest.mark.parametrize("gate", [False, True])
def test_experts_product(T, M, E, N, K, gate):
    g = _gen(T + 3 * M + E + N + K)
    N = 2 * N if gate else N
    X, W, sX, sW = _codes(g, T, K), _codes(g, E, N, K), _scales(g, T), _scales(g, E, N)
    if gate:
        sW /= 64 * K ** 0.5                              # gates of a size whose slope is not all at its ends
    rows = None if T == M else torch.randint(0, T, (M,), generator=g, dtype=torch.int32)
    off = _split(M, E, M, first=3 if M > 100 else 0, last=5 if M > 100 else 1)
    _say("experts", T, M, E, N, K, gate)
    call = dbs.gemm_moe_swiglu_i8 if gate else dbs.gemm_moe_i8
    D = call(X.cuda(), sX.cuda(), W.cuda(), sW.cuda(), torch.tensor(off, dtype=torch.int32).cuda(),
             None if rows is None else rows.cuda())
    h = _i8.moe_product(*(_moe.f64(t) for t in (X, sX, W, sW)), off, None if rows is None else rows.numpy())
    got = _moe.f64(D)
    if gate:
        a, u = h[:, : N // 2], h[:, N // 2:]
        assert np.all(np.abs(got - _i8.silu(a) * u) <= _i8.gate_bound(a, u, _i8.scaled_bound(a), _i8.scaled_bound(u)))
    else:
        assert np.all(np.abs(got - h) <= _i8.product_bound(h, True))
    assert not got[: off[0]].any() and not got[off[-1]:].any()


def test_experts_rows_and_offsets_out_of_range():
    """Row indices outside X stand for zero rows; offsets are clamped and made ascending."""
    g = _gen(2)
    T, M, E, N, K = 20, 300, 4, 72, 96
    X, W, sX, sW = _codes(g, T, K), _codes(g, E, N, K), _scales(g, T), _scales(g, E, N)
    rows = torch.randint(0, T, (M,), generator=g, dtype=torch.int32)
    rows[::7], rows[1::7], rows[2::7] = -1, T, 2 ** 31 - 1
    D = dbs.gemm_moe_i8(X.cuda(), sX.cuda(), W.cuda(), sW.cuda(),
                        torch.tensor([-5, 100, 60, 250, 1000], dtype=torch.int32).cuda(), rows.cuda())
    want = _i8.moe_product(*(_moe.f64(t) for t in (X, sX, W, sW)), [0, 100, 100, 250, 300], rows.numpy())
    assert np.all(np.abs(_moe.f64(D) - want) <= _i8.product_bound(want, True))


# Groups whose rows make more tiles than their number leads to expect, so that
# workgroups of the small tiles take several: group sizes, N, K
RAGGED = [([17, 1] * 4, 1024, 336), ([17, 0, 33, 2] * 4, 700, 1040), ([65] * 4, 640, 2048), ([65] * 4, 1300, 1040),
          ([1, 129, 0, 70, 64, 3], 1500, 272), ([5, 16, 0, 20, 31, 1, 9] * 3, 2050, 400)]


@pytest.mark.parametrize("sizes,N,K", RAGGED)
@pytest.mark.parametrize("gate", [False, True])
def test_experts_with_more_tiles_than_expected(sizes, N, K, gate):
    E, M = len(sizes), sum(sizes)
    g = _gen(M + N)
    X, W, sX, sW = _codes(g, 90, K), _codes(g, E, N, K), _scales(g, 90), _scales(g, E, N) / (64 * K ** 0.5)
    rows = torch.randint(0, 90, (M,), generator=g, dtype=torch.int32)
    off = np.concatenate([[0], np.cumsum(sizes)])
    call = dbs.gemm_moe_swiglu_i8 if gate else dbs.gemm_moe_i8
    args = [t.cuda() for t in (X, sX, W, sW, torch.tensor(off, dtype=torch.int32), rows)]
    _say("ragged", sizes, N, K, gate)
    D = call(*args)
    h = _i8.moe_product(*(_moe.f64(t) for t in (X, sX, W, sW)), off, rows.numpy())
    if gate:
        a, u = h[:, : N // 2], h[:, N // 2:]
        assert np.all(np.abs(_moe.f64(D) - _i8.silu(a) * u) <= _i8.gate_bound(a, u, _i8.scaled_bound(a), _i8.scaled_bound(u)))
    else:
        assert np.all(np.abs(_moe.f64(D) - h) <= _i8.product_bound(h, True))
    with dbs.using_library(dbs.load_poison_library()):
        assert torch.equal(call(*args), D)


@pytest.mark.parametrize("M", [1, 30, 200, 700, 3000])
def test_experts_of_one_group_are_the_dense_product(M):
    """The same numbers whichever tiles: sums are whole."""
    g = _gen(M)
    A, B, sA, sB = (t.cuda() for t in (_codes(g, M, 320), _codes(g, 600, 320), _scales(g, M), _scales(g, 600)))
    off = torch.tensor([0, M], dtype=torch.int32).cuda()
    assert torch.equal(dbs.gemm_moe_i8(A, sA, B[None], sB[None], off), dbs.gemm_i8(A, sA, B, sB))


# --------------------------------------------------------------- where it runs


def _layer(x, logits, q13, s13, q2, s2, bias, k=4):
    """A routed layer served in 8-bit integers, every call of it."""
    r = dbs.moe_route_grouped(logits, k, bias, groups=4, kept_groups=2, scale=2.5)
    qx, sx = dbs.quant_i8(x)
    a = dbs.gemm_moe_swiglu_i8(qx, sx, q13, s13, r.offsets, r.rows)
    qa, sa = dbs.quant_i8(a)
    y = dbs.gemm_moe_i8(qa, sa, q2, s2, r.offsets)
    shared = dbs.gemm_i8(qx, sx, q13[0], s13[0])
    return [*r, qx, sx, a, qa, sa, y, dbs.moe_combine(y, r.slots, r.weights), shared]


def _layer_inputs(T, E=16, H=128, F=96, seed=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w13 = torch.randn(E * 2 * F, H, generator=g, device="cuda") * H ** -0.5
    w2 = torch.randn(E * H, F, generator=g, device="cuda") * F ** -0.5
    q13, s13 = dbs.quant_i8(w13)
    q2, s2 = dbs.quant_i8(w2)
    return (torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16),
            torch.randn(T, E, generator=g, device="cuda"), q13.view(E, 2 * F, H), s13.view(E, 2 * F), q2.view(E, H, F),
            s2.view(E, H), torch.randn(E, generator=g, device="cuda") * 0.1)


@pytest.mark.parametrize("T", [1, 100, 3000])
def test_graph_replays_on_new_inputs(T):
    args = _layer_inputs(T)
    x, logits = args[0], args[1]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _layer(*args)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _layer(*args)
    g = torch.Generator(device="cuda")
    for i in range(4):
        g.manual_seed(50 + i)
        x.copy_(torch.randn(x.shape, generator=g, device="cuda", dtype=x.dtype))
        logits.copy_(torch.randn(logits.shape, generator=g, device="cuda"))
        if i == 2:
            logits[::3] = -float("inf")
        graph.replay()
        want = _layer(*args)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", PARTS[:3])
def test_graph_of_two_launches(M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    codes = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)
    A, B, sA, sB = codes(M, K), codes(N, K), torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    out = torch.full((M, N), float("nan"), device="cuda", dtype=torch.bfloat16)
    dbs.gemm_i8(A, sA, B, sB)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dbs.gemm_i8(A, sA, B, sB, out=out)
    for _ in range(3):
        A.copy_(codes(M, K))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, dbs.gemm_i8(A, sA, B, sB))
        assert bool(torch.isfinite(got).all())


def test_other_streams_and_two_calls_at_once():
    args = _layer_inputs(700)
    other = _layer_inputs(900, seed=5)
    want, want2 = _layer(*args), _layer(*other)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(a):
            got = _layer(*args)
        with torch.cuda.stream(b):
            got2 = _layer(*other)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x, y) for x, y in zip(got2, want2))


# sizes that reach every kernel, with several tiles to a workgroup
POISON = [(3, 70000, 200), (900, 33000, 640), (5000, 6000, 400), (9000, 9000, 130), (1500, 2500, 1024), (700, 30000, 260), (2047, 4102, 400), (1100, 9000, 768), (64, 30000, 512),
          (64, 40000, 512), (2157, 6150, 1040), (16, 40000, 1024), (250, 8000, 2064)]


@pytest.mark.parametrize("M,N,K", POISON)
def test_poison_build_gives_the_same_bits(M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    K = K // 16 * 16
    A = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sA, sB = (torch.rand(n, generator=g, device="cuda") + 0.1 for n in (M, N))
    rows = torch.randint(0, M, (M,), generator=g, device="cuda", dtype=torch.int32)
    off = torch.tensor([0, M // 3, M // 3, M - M // 5], device="cuda", dtype=torch.int32)
    W = torch.stack([B[: 2 * (N // 8)]] * 3)
    sW = torch.rand(3, W.shape[1], generator=g, device="cuda") * 1e-3

    def calls():
        return (dbs.gemm_i8(A, sA, B, sB), dbs.gemm_i8(A, sA, B, sB, out_dtype=torch.float32),
                dbs.gemm_moe_i8(A, sA, W, sW, off, rows), dbs.gemm_moe_i8(A, sA, W, sW, off),
                dbs.gemm_moe_swiglu_i8(A, sA, W, sW, off, rows))

    _say("poison", M, N, K)
    want = calls()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(calls(), want))
    with dbs.using_library(dbs.load_poison_library()):
        got = calls()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # (and they are right, on a sample of rows and columns)
    r = torch.randint(0, M, (40,), generator=g, device="cuda")
    c = torch.randint(0, N, (40,), generator=g, device="cuda")
    D = _i8.product(*(_moe.f64(t) for t in (A[r], sA[r], B[c], sB[c])))
    assert np.all(np.abs(_moe.f64(want[1][r][:, c]) - D) <= _i8.product_bound(D, False))


def test_outputs_beyond_4_gib():
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    M, N, K = 1_100_003, 2048, 32
    A = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sA, sB = (torch.rand(n, generator=g, device="cuda") for n in (M, N))
    _say("gemm", M, N, K)
    D = dbs.gemm_i8(A, sA, B, sB, out_dtype=torch.float32)
    r = torch.tensor([0, 1, 262143, 262144, 524_288, 700_000, M - 1], device="cuda")
    want = _i8.product(*(_moe.f64(t) for t in (A[r], sA[r], B, sB)))
    assert np.all(np.abs(_moe.f64(D[r]) - want) <= _i8.product_bound(want, False))
    q, s = dbs.quant_i8(D)
    codes, _ = _i8.quant(_moe.f64(D[r]))
    assert np.array_equal(q[r].cpu().numpy(), codes)


# ------------------------------------------------------------------ the example


def _example():
    import importlib.util
    from pathlib import Path

    path = Path(__file__).resolve().parent.parent / "examples" / "moe_layer_i8.py"
    spec = importlib.util.spec_from_file_location("moe_layer_i8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,experts,groups,k", [(1, 8, 4, 2), (200, 16, 4, 3), (1500, 32, 8, 4)])
def test_example_layer(tokens, experts, groups, k):
    """Quantising a row is off by amax / 127 / 12^0.5 (rms): 1.4 % with a largest value of six
    deviations.  Through the gate, a product of two, that is at most three per cent, the gate's own
    rows (ten deviations) add 2.3 %: below 6 % together."""
    far = _example().run(tokens, 256, 128, experts, groups, k)
    for name, v in far.items():
        if name != "router gradient, norm":
            assert v < 0.06, (name, v)
    assert np.isfinite(far["router gradient, norm"]) and far["router gradient, norm"] > 0


def test_example_router_gradient():
    """Against the formula in 64 bits, through the layer's own rows."""
    m = _example()
    torch.manual_seed(1)
    layer = m.MoeLayerI8(64, 32, 16, 4, 3)
    x = torch.randn(40, 64, device="cuda", dtype=torch.bfloat16)
    target = torch.randn(40, 64, device="cuda")
    layer.router_loss(x, target).backward()
    r = layer.route(x)
    y = _moe.f64(layer.rows(x, r))[r.slots.cpu().numpy()]                       # (T, k, H); every token has k
    w = _moe.f64(r.weights)
    out = (w[..., None] * y).sum(1)
    dw = (2 * (out - _moe.f64(target))[:, None, :] * y).sum(-1) / out.size
    logits = _moe.f64(x.float() @ layer.router)
    dlogits = _i8.grouped_grad(logits, r.experts.cpu().numpy(), dw, "sigmoid", True, layer.scale)
    want = _moe.f64(x).T @ dlogits
    # fp32 throughout: sums of 64 and 40 terms, a few dozen roundings of each
    assert np.all(np.abs(_moe.f64(layer.router.grad) - want) <= 200 * 2.0 ** -23 * (np.abs(_moe.f64(x)).T @ np.abs(dlogits) + np.abs(dlogits).max()))


def test_example_has_no_second_derivative():
    m = _example()
    layer = m.MoeLayerI8(64, 32, 8, 2, 2)
    x = torch.randn(4, 64, device="cuda", dtype=torch.bfloat16)
    loss = layer.router_loss(x, torch.zeros(4, 64, device="cuda"))
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(loss, layer.router, create_graph=True)
