"""The router by groups of experts on the GPU against its plain 64-bit form (-m
gpu)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _i8, _moe

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _say(*a):
    print(*a, flush=True)


def _logits(T, E, dtype, seed, closed):
    g = _gen(seed)
    x = torch.randn(T, E, generator=g) * 2
    if closed:
        x[torch.rand(T, E, generator=g) < closed] = -float("inf")
        x[::5] = -float("inf")                       # tokens without any open expert
    return x.to(dtype)


def _check(x, k, bias, groups, kept, best, scores, renorm, scale):
    r = dbs.moe_route_grouped(x.cuda(), k, None if bias is None else bias.cuda(), groups, kept, best, scores, renorm, scale)
    X = _moe.f64(x)
    experts = _i8.choose(X, k, None if bias is None else _moe.f64(bias), groups, kept, best, scores)
    offsets, rows, slots = _moe.routing(experts, x.shape[1])
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    w, steps = _i8.weights(X, experts, scores, renorm, np.float32(scale).astype(np.float64))
    # an exponential's argument is rounded once (half a step of its magnitude), the
    # exponentials, the sum of k, two divisions and the factor take a step or two each
    assert np.all(np.abs(_moe.f64(r.weights) - w) <= (20 + k + steps) * 2.0 ** -23 * np.abs(w) + 2.0 ** -126)
    return r


# T, E, k, groups, kept, best: every number of keys a lane holds, whole loads and
# not, groups of every number of lanes and of no power of two, tokens on both sides of 64 and 2048
ROUTE = [(1, 1, 1, 1, 1, 2), (1, 256, 8, 8, 4, 2), (3, 5, 5, 1, 1, 2), (63, 34, 4, 2, 1, 2), (64, 128, 8, 4, 2, 1),
         (65, 160, 6, 8, 3, 1), (200, 64, 16, 16, 4, 2), (130, 60, 3, 3, 2, 2), (90, 45, 7, 5, 2, 2), (77, 112, 8, 7, 7, 2),
         (40, 512, 8, 1, 1, 2), (33, 512, 10, 8, 4, 2), (31, 1024, 16, 1, 1, 1), (20, 1024, 4, 16, 3, 2),
         (66, 16, 1, 16, 1, 2), (50, 176, 8, 11, 5, 2), (70, 24, 2, 12, 6, 2), (300, 256, 8, 8, 4, 2), (100, 208, 5, 13, 2, 1)]


@pytest.mark.parametrize("T,E,k,groups,kept,best", ROUTE)
@pytest.mark.parametrize("dtype,scores,renorm,closed,bias", [
    (torch.float32, "sigmoid", True, 0.0, True), (torch.bfloat16, "sigmoid", False, 0.0, False),
    (torch.float32, "softmax", False, 0.5, True), (torch.bfloat16, "softmax", True, 0.0, True),
    (torch.bfloat16, "sigmoid", True, 0.85, True)])
def test_route(T, E, k, groups, kept, best, dtype, scores, renorm, closed, bias):
    x = _logits(T, E, dtype, T * 1000 + E, closed)
    b = torch.randn(E, generator=_gen(E)) * 0.3 if bias else None
    _say("route", T, E, k, groups, kept, best, dtype, scores, renorm, closed)
    _check(x, k, b, groups, kept, best, scores, renorm, 2.5)


# 16, 32 and 64 tokens to a workgroup on both sides of each switch, counts of one and of several threads a row
@pytest.mark.parametrize("T,E,k,groups,kept", [(2048, 32, 4, 4, 2), (2049, 48, 4, 8, 4), (4500, 160, 6, 8, 3), (4096, 17, 3, 1, 1),
                                               (8192, 24, 16, 2, 2), (8193, 3, 2, 1, 1), (16384, 20, 2, 4, 3),
                                               (16385, 36, 3, 4, 2), (1100, 1024, 4, 8, 4), (600, 520, 5, 1, 1)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_route_of_many_tokens(T, E, k, groups, kept, scores):
    x = _logits(T, E, torch.float32, T, 0.3)
    _check(x, k, torch.randn(E, generator=_gen(2)), groups, kept, 2, scores, True, 1.0)


def test_ties_go_to_the_lower_expert_and_group():
    x = torch.zeros(5, 16)
    x[1, 8:] = 1.0                                     # groups 2 and 3 above 0 and 1
    x[2, [3, 7, 11, 15]] = 2.0                         # every group's best the same
    x[3, ::2] = -1.0
    r = _check(x, 4, None, 4, 2, 2, "sigmoid", True, 1.0)
    assert r.experts.cpu().tolist()[:3] == [[0, 1, 2, 3], [8, 9, 10, 11], [3, 7, 0, 1]]
    # the bias decides, and below zero too
    b = torch.full((16,), -4.0)
    b[5] = -3.0
    r = _check(x[:1], 3, b, 4, 2, 2, "sigmoid", True, 1.0)
    assert r.experts.cpu().tolist() == [[5, 0, 1]]      # group 1, then group 0 of three that tie


def test_scores_nearer_than_fp32_tells_apart():
    """Choices between scores that are one and the same in fp32."""
    x = torch.tensor([[16.0, 16.0 + 2.0 ** -19, 17.0, -1.0]])
    assert torch.sigmoid(x[0, 0]) == torch.sigmoid(x[0, 1])
    r = _check(x, 3, None, 1, 1, 2, "sigmoid", False, 1.0)
    assert r.experts.cpu().tolist() == [[2, 1, 0]]
    bias = torch.tensor([0.5, 0.5, 0.0, 0.0])
    assert _check(x, 2, bias, 2, 1, 2, "sigmoid", False, 1.0).experts.cpu().tolist() == [[1, 0]]


def test_special_logits():
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    x = torch.tensor([[1.0, inf, inf, 0.0, -1.0, 2.0],
                      [nan, 1.0, nan, 2.0, -inf, nan],
                      [low, low, low, low, low, low],
                      [nan, nan, nan, -inf, -inf, -inf],
                      [-300.0, -200.0, -250.0, -260.0, -inf, -400.0],   # scores below fp32's range
                      [90.0, 80.0, 100.0, 85.0, 30.0, 20.0]])
    for scores in ("sigmoid", "softmax"):
        for renorm in (True, False):
            # (fp64 has no scores for the third row's logits: all tie)
            _check(x, 3, None, 1, 1, 2, scores, renorm, 1.0)
    r = dbs.moe_route_grouped(x.cuda(), 3, torch.tensor([0.0, -inf, nan, 0.0, inf, 0.0]).cuda())
    # closed by their bias: 1 and 2; 4's is the largest, where its logit is open
    assert r.experts.cpu().tolist() == [[4, 5, 0], [3, -1, -1], [4, 0, 3], [-1, -1, -1], [3, 0, 5], [4, 0, 3]]
    assert torch.isfinite(r.weights).all()


def test_groups_without_open_experts_are_not_kept():
    inf = float("inf")
    x = torch.tensor([[-inf, -inf, 1.0, -inf, -inf, -inf, 0.5, 0.25]])
    r = _check(x, 4, None, 4, 3, 2, "sigmoid", True, 1.0)
    assert r.experts.cpu().tolist() == [[2, 6, 7, -1]]
    # one open expert above another group's two: 0.9 against 0.1 + 0.1
    b = torch.tensor([0.0, 0.0, 0.0, 0.0])
    r = _check(torch.tensor([[-2.2, -2.2, 2.2, -inf]]), 1, b, 2, 1, 2, "sigmoid", True, 1.0)
    assert r.experts.cpu().tolist() == [[2]]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (33, 160, 6), (100, 17, 4), (17, 1024, 16), (50, 300, 8), (600, 256, 8)])
@pytest.mark.parametrize("dtype,scores,renorm,closed", [
    (torch.float32, "sigmoid", True, 0.0), (torch.bfloat16, "sigmoid", False, 0.0), (torch.float32, "sigmoid", False, 0.6),
    (torch.bfloat16, "sigmoid", True, 0.8), (torch.float32, "softmax", True, 0.0), (torch.bfloat16, "softmax", False, 0.5)])
def test_backward(T, E, k, dtype, scores, renorm, closed):
    x = _logits(T, E, dtype, T + E, closed)
    d = torch.randn(T, k, generator=_gen(5))
    experts = _i8.choose(_moe.f64(x), k, None, 1, 1, 2, scores)
    got = _moe.f64(dbs.moe_route_grouped_backward(x.cuda(), torch.tensor(experts, dtype=torch.int32).cuda(), d.cuda(),
                                                  scores=scores, renormalize=renorm, scale=1.75))
    want = _i8.grouped_grad(_moe.f64(x), experts, _moe.f64(d), scores, renorm, 1.75)
    # weights to (E + 28) steps (softmax) or k + 28, the inner sum over terms of at most |d|
    n = E if scores == "softmax" else k
    bound = (2 * n + 60) * 2.0 ** -23 * 1.75 * float(d.abs().max())
    if dtype == torch.bfloat16:
        bound = bound + _moe.HALF_STEP * np.abs(want)
    assert np.all(np.abs(got - want) <= bound)
    if scores == "sigmoid":
        on = np.zeros((T, E), dtype=bool)
        for t in range(T):
            on[t, experts[t][experts[t] >= 0]] = True
        assert not got[~on].any()


def test_backward_of_small_and_saturated_scores():
    x = torch.tensor([[-90.0, -100.0, -95.0, 3.0], [50.0, 60.0, 40.0, 0.0], [-1e30, -2e30, -1e30, 1.0],
                      [float("nan"), 1.0, -float("inf"), 2.0]])
    e = torch.tensor([[0, 1, 2], [1, 0, 2], [0, 2, 1], [3, 1, -1]], dtype=torch.int32)
    d = torch.tensor([[1.0, -2.0, 0.5]]).repeat(4, 1)
    for renorm in (True, False):
        got = _moe.f64(dbs.moe_route_grouped_backward(x.cuda(), e.cuda(), d.cuda(), renormalize=renorm))
        want = _i8.grouped_grad(_moe.f64(x), e.numpy(), _moe.f64(d), "sigmoid", renorm, 1.0)
        assert np.all(np.isfinite(got))
        # relative steps of the factors (exponents up to 100) and of the inner sum
        assert np.all(np.abs(got - want) <= 140 * 2.0 ** -23 * (np.abs(want) + (2.5 * np.abs(want) if renorm else 0)) + 2.0 ** -126)


def test_gradient_against_differences():
    T, E, k, h = 5, 16, 3, 2.0 ** -7
    x = torch.randn(T, E, generator=_gen(11))
    d = torch.randn(T, k, generator=_gen(12))
    bias = torch.randn(E, generator=_gen(13))
    for scores in ("sigmoid", "softmax"):
        for renorm in (True, False):
            args = dict(groups=4, kept_groups=2, scores=scores, renormalize=renorm, scale=1.5)
            r = dbs.moe_route_grouped(x.cuda(), k, bias.cuda(), **args)
            g = _moe.f64(dbs.moe_route_grouped_backward(x.cuda(), r.experts, d.cuda(), scores, renorm, 1.5))
            for t in range(T):
                for e in range(E):
                    ends = []
                    for s in (h, -h):
                        y = x.clone()
                        y[t, e] += s
                        q = dbs.moe_route_grouped(y.cuda(), k, bias.cuda(), **args)
                        if not torch.equal(q.experts, r.experts):
                            break                     # the choice changes here: no derivative
                        ends.append(float((_moe.f64(q.weights)[t] * _moe.f64(d)[t]).sum()))
                    if len(ends) == 2:
                        # third derivatives of the weights are below 2, fp32 weights to 40 steps of 2
                        assert abs((ends[0] - ends[1]) / (2 * h) - g[t, e]) <= 6 * h * h * 4 + 240 * 2.0 ** -23 / h


def test_softmax_without_groups_agrees_with_moe_route():
    x = _logits(500, 96, torch.float32, 3, 0.4)
    for renorm in (True, False):
        a, b = dbs.moe_route(x.cuda(), 4, renorm), dbs.moe_route_grouped(x.cuda(), 4, scores="softmax", renormalize=renorm)
        assert all(torch.equal(s, t) for s, t in zip((a[0], *a[2:]), (b[0], *b[2:])))
        assert torch.allclose(a.weights, b.weights, rtol=100 * 2.0 ** -23, atol=0)


def test_repeats_bit_for_bit():
    x = _logits(5000, 256, torch.float32, 3, 0.0).cuda()
    b = torch.randn(256, generator=_gen(2)).cuda() * 0.1
    want = dbs.moe_route_grouped(x, 8, b, 8, 4, scale=2.5)
    for _ in range(5):
        assert all(torch.equal(s, t) for s, t in zip(dbs.moe_route_grouped(x, 8, b, 8, 4, scale=2.5), want))
