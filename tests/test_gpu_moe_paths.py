"""The mixture-of-experts operators where it is the path that can go wrong
(-m gpu): outputs beyond 4 GiB, HIP graphs, the LDS-poison build against the
product build, repeated calls, the example's layer."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _moe

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _cuda_gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def _say(*a):
    print(*a, flush=True)


def _check_rows(x, w, got, K, mn=False):
    """Sampled output rows: x (n, K), w (N, K) or (K, N) of their expert."""
    X, W = _moe.f64(x), _moe.f64(w)
    W = W if mn else W.T
    D, S = X @ W, np.abs(X) @ np.abs(W)
    assert np.all(np.abs(_moe.f64(got) - D) <= _moe.product_bound(D, S, K))


def test_outputs_beyond_4_gib():
    M, E, N, K = 1_100_003, 3, 2048, 64
    g = _cuda_gen(1)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    W = torch.randn(E, N, K, generator=g, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 700_001, 1_000_000, 1_099_990], dtype=torch.int32).cuda()
    _say("product", M, E, N, K)
    D = dbs.gemm_moe_bf16(X, W, off)
    for e, r in ((0, [0, 1, 524_288, 700_000]), (1, [700_001, 999_999]), (2, [1_000_000, 1_048_600, 1_099_989])):
        _check_rows(X[r], W[e], D[r], K)
    assert bool((D[1_099_990:] == 0).all())
    del D
    _say("gated", M, E, N, K)
    W2 = torch.randn(E, 2 * N, K, generator=g, device="cuda", dtype=torch.bfloat16) * 0.2
    D = dbs.gemm_moe_swiglu_bf16(X, W2, off)
    r = [1_000_000, 1_060_001, 1_099_989]
    h, S = _moe.f64(X[r]) @ _moe.f64(W2[2]).T, np.abs(_moe.f64(X[r])) @ np.abs(_moe.f64(W2[2])).T
    acc = K * 2.0 ** -23 * S
    a, u = h[:, :N], h[:, N:]
    assert np.all(np.abs(_moe.f64(D[r]) - _moe.silu(a) * u) <= _moe.gate_bound(a, u, acc[:, :N], acc[:, N:]))
    _say("combine and its gradient over", M, "rows")
    T = M // 1                                         # one row per token
    slots = torch.randperm(M, generator=g, device="cuda").to(torch.int32).view(T, 1)
    out = dbs.moe_combine(D, slots)
    assert torch.equal(out[r], D[slots[r, 0].long()])
    w = torch.rand(T, 1, generator=g, device="cuda")
    end = torch.tensor([0, M], dtype=torch.int32).cuda()
    dY, dw = dbs.moe_combine_backward(out, D, slots, w, end)
    at = slots[r, 0].long()
    assert torch.equal(dY[at], (w[r] * out[r].float()).to(torch.bfloat16))


def test_dw_beyond_4_gib():
    E, N, K, M = 40, 4096, 8192, 400
    g = _cuda_gen(2)
    X = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    dY = torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * 10
    _say("dw", E, N, K, M)
    d = dbs.gemm_moe_dw_bf16(dY, X, off, out_dtype=torch.float32)
    for e in (0, 31, 39):
        a, b = _moe.f64(dY[10 * e:10 * e + 10, 4000:]), _moe.f64(X[10 * e:10 * e + 10, 8000:])
        want, size = a.T @ b, np.abs(a).T @ np.abs(b)
        assert np.all(np.abs(_moe.f64(d[e, 4000:, 8000:]) - want) <= 11 * 2.0 ** -23 * size)


def test_graph_replays_on_new_inputs():
    """Router, products, sums and their gradients captured once; every replay
    against the eager calls, with eager work in between."""
    T, E, k, H, F = 100, 16, 4, 128, 64
    g = _cuda_gen(3)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    w13 = torch.randn(E, 2 * F, H, generator=g, device="cuda", dtype=torch.bfloat16) * 0.1
    w2 = torch.randn(E, H, F, generator=g, device="cuda", dtype=torch.bfloat16) * 0.1

    def step():
        r = dbs.moe_route(logits, k)
        h = dbs.gemm_moe_bf16(x, w13, r.offsets, r.rows)
        a = dbs.swiglu(h)
        y = dbs.gemm_moe_bf16(a, w2, r.offsets)
        out = dbs.moe_combine(y, r.slots, r.weights)
        dy, dweights = dbs.moe_combine_backward(out, y, r.slots, r.weights, r.offsets)
        dh = dbs.swiglu_backward(dbs.gemm_moe_bf16(dy, w2, r.offsets, lw=dbs.MN_MAJOR), h)
        return [*r, out, dweights, dbs.gemm_moe_dw_bf16(dh, x, r.offsets, r.rows),
                dbs.moe_route_backward(logits, r.experts, dweights)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(4):
        x.copy_(torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16))
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


CASES = [(300, 700, 4, 264, 136), (2000, 5000, 3, 520, 328), (48, 300, 64, 96, 200), (700, 1500, 5, 776, 1032),
         (2500, 2500, 2, 512, 256),
         # 256-row tiles in every form, and 64 x 128 tiles of dW over several rounds
         (1500, 2600, 3, 4400, 2312), (3000, 3000, 7, 4096, 2120), (900, 12000, 60, 320, 1544),
         # 128-row tiles: K-major, and of the last MN-major and gated
         (900, 2048, 2, 2056, 200), (2000, 2900, 2, 2056, 1544)]


def _inputs(T, M, E, N, K, seed):
    g = _gen(seed)
    X = _bf16(g, T, K).cuda()
    W = _bf16(g, E, N, K).cuda()
    dY = _bf16(g, M, N).cuda()
    cuts = np.sort(np.random.default_rng(seed).integers(0, M + 1, E - 1))
    off = torch.tensor(np.concatenate([[0], cuts, [M]]), dtype=torch.int32).cuda()
    rows = torch.randint(0, T, (M,), generator=g, dtype=torch.int32).cuda()
    return X, W, dY, off, rows


def _all(X, W, dY, off, rows):
    out = [dbs.gemm_moe_bf16(X, W, off, rows), dbs.gemm_moe_swiglu_bf16(X, W, off, rows),
           dbs.gemm_moe_bf16(dY, W, off, lw=dbs.MN_MAJOR), dbs.gemm_moe_dw_bf16(dY, X, off, rows),
           dbs.gemm_moe_dw_bf16(dY, X, off, rows, out_dtype=torch.float32)]
    if X.shape[0] == rows.shape[0]:
        out += [dbs.gemm_moe_bf16(X, W, off), dbs.gemm_moe_dw_bf16(dY, X, off)]
    return out


@pytest.mark.parametrize("T,M,E,N,K", CASES)
def test_poison_build_gives_the_same_bits(T, M, E, N, K):
    """Every direct-to-LDS load's destination filled with NaN before the load:
    a read ahead of its load, or a refill ahead of a read, would show."""
    a = _inputs(T, M, E, N, K, N + K)
    _say("poison", T, M, E, N, K)
    want = _all(*a)
    with dbs.using_library(dbs.load_poison_library()):
        got = _all(*a)
    for u, v in zip(got, want):
        assert torch.equal(u, v)


@pytest.mark.parametrize("T,M,E,N,K", CASES[:3] + CASES[5:])
def test_calls_repeat_bit_for_bit(T, M, E, N, K):
    a = _inputs(T, M, E, N, K, N)
    want = _all(*a)
    for _ in range(20):
        for u, v in zip(_all(*a), want):
            assert torch.equal(u, v)


def test_one_row_has_the_same_bits_in_any_company():
    """A row's product does not depend on its group's other rows."""
    g = _gen(7)
    E, N, K = 4, 160, 256
    X, W = _bf16(g, 4000, K).cuda(), _bf16(g, E, N, K).cuda()
    few = torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32).cuda()
    a = dbs.gemm_moe_bf16(X, W, few, torch.tensor([5, 6, 7, 8], dtype=torch.int32).cuda())
    b = dbs.gemm_moe_bf16(X, W, torch.tensor([0, 1, 1, 1, 1], dtype=torch.int32).cuda(),
                          torch.tensor([5], dtype=torch.int32).cuda())
    assert torch.equal(a[0], b[0])
    whole = torch.tensor([0, 4000, 4000, 4000, 4000], dtype=torch.int32).cuda()
    c = dbs.gemm_moe_bf16(X, W, whole)
    d = dbs.gemm_moe_bf16(X[:3001].contiguous(), W, torch.tensor([0, 3001, 3001, 3001, 3001], dtype=torch.int32).cuda())
    assert torch.equal(c[:3001], d)


def test_one_row_has_the_same_bits_in_any_company_under_large_tiles():
    g = _gen(9)
    E, N, K = 2, 4360, 72
    X, W = _bf16(g, 1400, K).cuda(), _bf16(g, E, N, K).cuda()
    o = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()
    a = dbs.gemm_moe_bf16(X, W, o(0, 1400, 1400))
    b = dbs.gemm_moe_bf16(X[:1301].contiguous(), W, o(0, 1301, 1301))
    assert torch.equal(a[:1301], b)
    c = dbs.gemm_moe_bf16(X, W, o(0, 1400, 1400), torch.arange(1399, -1, -1, dtype=torch.int32).cuda())
    assert torch.equal(c.flip(0), a)


def test_offsets_that_are_no_offsets_stay_inside():
    """Descending, negative and too large offsets are clamped and read as
    empty groups; the call ends and writes only D."""
    g = _gen(8)
    M, E, N, K = 300, 5, 72, 64
    X, W, dY = _bf16(g, M, K).cuda(), _bf16(g, E, N, K).cuda(), _bf16(g, M, N).cuda()
    off = [-7, 50, 20, 120, 10_000, 60]              # read as 0, 50, 50, 120, 300, 300
    read = [0, 50, 50, 120, 300, 300]
    o = torch.tensor(off, dtype=torch.int32).cuda()
    r = torch.tensor(read, dtype=torch.int32).cuda()
    rows = torch.arange(M, dtype=torch.int32).cuda()
    for u, v in zip(_all(X, W, dY, o, rows), _all(X, W, dY, r, rows)):
        assert torch.equal(u, v)
    few = dbs.gemm_moe_bf16(X[:8].contiguous(), W, torch.tensor([3, -1, 2, 9, 5, 8], dtype=torch.int32).cuda())
    assert torch.equal(few, dbs.gemm_moe_bf16(X[:8].contiguous(), W,
                                              torch.tensor([3, 3, 3, 8, 8, 8], dtype=torch.int32).cuda()))


@pytest.mark.parametrize("k", [1 << 40, 9, 0, -1, -(1 << 40)])
def test_route_refuses_k_without_sizing_outputs_by_it(k):
    x = torch.zeros(4, 8, device="cuda")
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(dbs.DbsError):
        dbs.moe_route(x, k)
    assert torch.cuda.max_memory_allocated() - before <= 1 << 16


def test_example_layer():
    """The layer's results against its plain form in 32 bits: intermediate
    rounding to bf16 (2^-8 each, five in a row at most in a gradient) keeps them
    within 5 * 2^-8 of each other."""
    import importlib.util
    from pathlib import Path

    path = Path(__file__).resolve().parent.parent / "examples" / "moe_layer.py"
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    far = m.run(512, 256, 128, 16, 4)
    _say(far)
    assert all(v <= 5 * 2.0 ** -8 for v in far.values())


def _example():
    import importlib.util
    from pathlib import Path

    path = Path(__file__).resolve().parent.parent / "examples" / "moe_layer.py"
    spec = importlib.util.spec_from_file_location("moe_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("loss", [lambda out: out.float().sum(), lambda out: out.float().square().sum()])
def test_example_layer_has_no_second_derivative(loss):
    """A gradient's gradient is an error, not the gradient of a constant."""
    layer = _example().MoeLayer(64, 32, 4, 2)
    x = torch.randn(8, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        torch.autograd.grad(loss(layer(x)), x, create_graph=True)
    torch.autograd.grad(loss(layer(x)), x)


@pytest.mark.parametrize("need", ["x", "router", "w13", "w2"])
def test_example_layer_computes_the_gradients_that_are_needed(need, monkeypatch):
    """One at a time: the same bits as with all of them, and no matrices'
    gradients where the matrices are frozen."""
    m = _example()
    torch.manual_seed(1)
    layer = m.MoeLayer(128, 64, 8, 2)
    x = torch.randn(40, 128, device="cuda", dtype=torch.bfloat16)
    leaves = {"x": x.requires_grad_(), "router": layer.router, "w13": layer.w13, "w2": layer.w2}
    dout = torch.randn_like(x)
    layer(x).backward(dout)
    want = {n: t.grad.clone() for n, t in leaves.items()}
    calls = []
    dw = m.dbs.gemm_moe_dw_bf16
    monkeypatch.setattr(m.dbs, "gemm_moe_dw_bf16", lambda *a, **k: calls.append(1) or dw(*a, **k))
    for n, t in leaves.items():
        t.grad = None
        t.requires_grad_(n == need)
    layer(x).backward(dout)
    assert torch.equal(leaves[need].grad, want[need])
    assert all(t.grad is None for n, t in leaves.items() if n != need)
    assert len(calls) == (need in ("w13", "w2"))
